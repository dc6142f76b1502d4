"""GPU: a call whose workspace cannot be had reports the error itself, and the thread's next call is
not blamed for it.

The failing call is made on a stream whose capture has been invalidated (by a synchronisation, which
a capturing stream refuses): the allocation is refused on the host, and nothing runs on the device.
"""
import ctypes

import pytest
import torch

import attention_forward_tiled_b200 as attn

pytestmark = pytest.mark.gpu

RELAXED = 2  # CU_STREAM_CAPTURE_MODE_RELAXED


def rand(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(1)).half().cuda()


def window_token():
    q, kv = rand(1, 1, 4, 64), rand(1, 2000, 2, 64)
    out, lse = torch.empty_like(q), torch.empty(1, 4, 1, device="cuda")
    return lambda s: attn.attn_fwd_window(q, kv, kv, 1500, 2, out=out, lse=lse, stream=s)


def window_gradients():
    q, kv = rand(1, 200, 4, 64), rand(1, 200, 2, 64)
    o, lse = attn.attn_fwd_window(q, kv, kv, 50)
    bufs = [torch.empty_like(t) for t in (q, kv, kv)]
    return lambda s: attn.attn_bwd_window(q, kv, kv, o, lse, q, 50, dq=bufs[0], dk=bufs[1], dv=bufs[2], stream=s)


def dense_token():
    q, kv = rand(1, 1, 4, 64), rand(1, 4000, 4, 64)
    out, lse = torch.empty_like(q), torch.empty(1, 4, 1, device="cuda")
    return lambda s: attn.attn_fwd(q, kv, kv, out=out, lse=lse, stream=s, path="decode", splits=4)


def dense_gradients():
    q = rand(1, 200, 4, 64)
    o, lse = attn.attn_fwd(q, q, q)
    bufs = [torch.empty_like(q) for _ in range(3)]
    return lambda s: attn.attn_bwd(q, q, q, o, lse, q, dq=bufs[0], dk=bufs[1], dv=bufs[2], stream=s)


@pytest.mark.parametrize("make", [window_token, window_gradients, dense_token, dense_gradients])
def test_a_failed_call_leaves_no_error_behind(make):
    call, good = make(), rand(1, 100, 2, 64)
    want = attn.attn_fwd(good, good, good)[0]
    call(None)  # kernels, limits and pools are set up by now
    torch.cuda.synchronize()
    cuda, stream = ctypes.CDLL("libcuda.so.1"), torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
    assert cuda.cuStreamBeginCapture_v2(handle, RELAXED) == 0
    try:
        assert cuda.cuStreamSynchronize(handle) != 0
        with pytest.raises(attn.AttnError) as failed:
            call(stream)
    finally:
        assert cuda.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0
    assert failed.value.code == attn.ATTN_ERR_CUDA
    assert torch.equal(attn.attn_fwd(good, good, good)[0], want)
    call(stream)
    assert attn.get_status(stream) == 0
