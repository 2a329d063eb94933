"""Tensors of another device than the call's are refused: the kernels get bare addresses.  The tensors here
lie on the host and only say that they are on a GPU; no call reaches a kernel."""
import pytest
import torch

import gather_qsa_pool_gb300 as qsa

H, D, PAGE, PAGES, V = 2, 16, 8, 4, 10
E4M3 = torch.float8_e4m3fn


class On(torch.Tensor):
    """A host tensor that says it is on GPU `gpu`."""
    gpu = 0

    def get_device(self):
        return self.gpu

    @property
    def is_cuda(self):
        return self.gpu >= 0


def on(t, gpu=0):
    t = t.as_subclass(On)
    t.gpu = gpu
    return t


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


@pytest.fixture
def cache(monkeypatch):
    pool = {n: on(torch.zeros(PAGES * PAGE, H, D)) for n in ("K", "V")}
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    return qsa.PagedCache(pool["K"], pool["V"], PAGE)


def every(call, tensors, **rest):
    """The call is refused with any one of the tensors on another GPU, or on the host."""
    for name in tensors:
        for gpu in (1, -1):
            args = {n: on(t, gpu if n == name else 0) for n, t in tensors.items()}
            with pytest.raises(ValueError, match="cuda:0|CUDA tensor|cuda:1"):
                call(**args, **rest)


def test_write(cache):
    every(lambda **a: qsa.paged_write(cache, **a),
          dict(table=i32(2, 2), cu_q=i32(3), kv_len=i32(2), k=torch.zeros(3, H, D), v=torch.zeros(3, H, D)))


def test_read(cache):
    every(lambda **a: qsa.paged_read(cache, **a),
          dict(table=i32(2, 2), kv_len=i32(2), n_cells=i32(2), K_out=torch.zeros(2, 5, H, D),
               V_out=torch.zeros(2, 5, H, D), pos=i32(2, 5), seq=i32(2)), max_cells=5)


def test_paged_attention(cache):
    every(lambda **a: qsa.paged_attn(cache, **a),
          dict(table=i32(2, 2), cu_q=i32(3), kv_len=i32(2), q=torch.zeros(3, 4, D), out=torch.zeros(3, 4, D),
               lse=torch.zeros(3, 4), workspace=torch.zeros(64, dtype=torch.uint8)), scale=1.0, max_q=1)


def test_prompt_attention():
    every(qsa.prompt_attn,
          dict(q=torch.zeros(3, 4, D), k=torch.zeros(3, H, D), v=torch.zeros(3, H, D), cu_seq=i32(3),
               out=torch.zeros(3, 4, D), lse=torch.zeros(3, 4), workspace=torch.zeros(64, dtype=torch.uint8)), scale=1.0)


def test_verification():
    every(qsa.draft_verify,
          dict(target=torch.zeros(2, 3, V), draft=torch.zeros(2, 2, V), tokens=i32(2, 2), u=torch.zeros(2, 3),
               tokens_out=i32(2, 3), n_accepted=i32(2), n_draft=i32(2)))


def test_a_cache_on_another_device_than_the_current(cache, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    args = [on(t) for t in (i32(2, 2), i32(3), i32(2), torch.zeros(3, H, D), torch.zeros(3, H, D))]
    with pytest.raises(ValueError, match="current device"):
        qsa.paged_write(cache, *args)


def test_a_stream_of_another_device(cache):
    class Stream:
        device_index, cuda_stream = 1, 0

    args = [on(t) for t in (i32(2, 2), i32(3), i32(2), torch.zeros(3, H, D), torch.zeros(3, H, D))]
    with pytest.raises(ValueError, match="a stream of cuda:1"):
        qsa.paged_write(cache, *args, stream=Stream())


def test_exponents_on_another_device():
    c = on(torch.zeros(PAGES * PAGE, H, D).to(E4M3))
    e = torch.zeros(PAGES * PAGE, H, dtype=torch.uint8)
    with pytest.raises(ValueError):
        qsa.PagedCache(c, c, PAGE, K_exp=on(e), V_exp=on(e, 1).to("meta"))
