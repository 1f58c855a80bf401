"""CPU tests of the write with norms: the oracle, and refusals that come before any HIP call."""
import ctypes

import numpy as np
import pytest
import torch

import heterogeneous_adapter_batching_amd as hl
import oracle
from test_attn_batch import DEVICE, cache, world  # noqa: F401
from test_attn_plan import _kv, _launch
from heterogeneous_adapter_batching_amd import attention


def write(L, kv, norm, **change):
    f = dict(q=0x1000, k=0x2000, v=0x3000, ldq=1024, ldk=256, ldv=256, rope=0x4000, q_out=0x5000, ld_out=1024,
             dtype=hl.LORA_F32, rope_len=20, rope_dim=128, reserved=0)
    f.update(change)
    n = dict(q=0x6000, k=0x7000, ld_q=0, ld_k=0, dtype=hl.LORA_F32, centred=0, eps=1e-6, reserved=0)
    n.update(norm or {})
    return hl._lib.lora_kv_write_norm(ctypes.byref(L), ctypes.byref(kv), ctypes.byref(hl.lora_kv_write_args_t(**f)),
                                      None if norm is None else ctypes.byref(hl.lora_head_norm_t(**n)), None)


@pytest.mark.parametrize("norm", [
    None, dict(q=None, k=None), dict(dtype=2), dict(dtype=-1), dict(eps=0.0), dict(eps=-1e-6), dict(eps=1.5),
    dict(eps=float("nan")), dict(centred=2), dict(ld_q=64), dict(ld_k=-128), dict(ld_q=132), dict(q=0x6008),
    dict(k=0x7004)])
def test_refuses_norms(norm):
    assert write(_launch(), _kv(), norm) == hl.LORA_EINVAL


def test_refuses_what_the_write_refuses():
    L, kv = _launch(), _kv()
    assert write(L, kv, {}, q=None, q_out=None) == hl.LORA_EINVAL  # a norm of a q that is not there
    assert write(L, kv, {}, k=None) == hl.LORA_EINVAL
    assert write(L, kv, {}, rope_len=19) == hl.LORA_EINVAL
    assert write(L, kv, {}, rope_dim=8) == hl.LORA_ESHAPE
    assert write(L, _kv(n_pages=3), {}) == hl.LORA_ESHAPE
    assert hl._lib.lora_kv_write_norm(ctypes.byref(L), ctypes.byref(kv), None, None, None) == hl.LORA_EINVAL


def test_an_empty_batch_launches_nothing():
    _, info = hl.lora_attn_plan(_launch().info.shape, [0], [0], None)
    assert write(hl.lora_attn_launch_t(0x1000, info), _kv(), {}, k=None, v=None) == hl.LORA_OK


def test_batch_refuses_weights(world):  # noqa: F811
    class Weights:
        def __init__(self, shape, dtype=torch.float32, device=DEVICE, step=1):
            self.shape, self.dtype, self.device, self.step = torch.Size(shape), dtype, device, step

        def dim(self):
            return len(self.shape)

        def stride(self, i):
            return self.step if i in (-1, self.dim() - 1) else self.shape[-1] * self.step

        def data_ptr(self):
            return 0x1000
    batch = attention.AttnBatch(cache(), 4)
    norm = batch._norm(Weights((64,)), Weights((2, 64)), 1e-5, True)
    assert (norm.ld_q, norm.ld_k, norm.dtype, norm.centred) == (0, 64, hl.LORA_F32, 1)
    norm = batch._norm(None, Weights((64,), torch.bfloat16), 1e-5, False)
    assert norm.q is None and norm.dtype == hl.LORA_BF16 and norm.centred == 0
    assert batch._norm(None, None, 1e-6, False) is None
    good = Weights((64,))
    for bad in (Weights((128,)), Weights((3, 64)), Weights((64,), torch.float16), Weights((64,), torch.bfloat16),
                Weights((64,), device=torch.device("cpu")), Weights((64,), step=2), Weights((1, 4, 64))):
        with pytest.raises(ValueError):
            batch._norm(good, bad, 1e-6, False)
        if bad.dtype != torch.bfloat16:
            with pytest.raises(ValueError):
                batch._norm(bad, None, 1e-6, False)


def test_oracle_norms_match_torch():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((5, 3, 64)) * 3 + 1, rng.standard_normal(64)
    t = torch.from_numpy(x)
    want = torch.nn.functional.layer_norm(t, (64,), torch.from_numpy(w), None, 1e-3)
    assert np.allclose(oracle.norm_ref(x, w, 1e-3, True), want.numpy(), rtol=1e-12)
    want = torch.nn.functional.rms_norm(t, (64,), torch.from_numpy(w), 1e-3)
    assert np.allclose(oracle.norm_ref(x, w, 1e-3, False), want.numpy(), rtol=1e-12)
    assert np.allclose(oracle.norm_ref([3.0, 4.0], 1.0, 0.0, False), np.array([3.0, 4.0]) / np.sqrt(12.5))
