"""CPU tests of the operators on token rows: the C ABI refuses bad arguments
before any CUDA call, the binding refuses host tensors, and the frequencies
follow their formulas."""
import ctypes
import math

import pytest
import torch

from submanifold_sparse_convolution_hash_gb300 import binding


@pytest.fixture(scope="module")
def libsc():
    from submanifold_sparse_convolution_hash_gb300 import build
    build.build()
    return binding.lib()


def attn(L, n_seq=1, t_q=4, t_k=4, hq=2, hk=2, d=64, scale=0.1, dtype=1, flags=0, ptr=None):
    return L.sc_attn_fwd(None, None, None, None, None, ptr, ptr, None, n_seq, t_q, t_k, hq, hk, d, scale, dtype, flags,
                         None)


@pytest.mark.parametrize("change,status", [
    (dict(flags=2), 1), (dict(dtype=7), 1), (dict(dtype=0), 5), (dict(n_seq=-1), 1), (dict(t_q=-1), 1),
    (dict(t_k=1 << 31), 1), (dict(hq=3), 1), (dict(hk=0), 1), (dict(hq=258, hk=2), 5), (dict(d=8), 5),
    (dict(d=100), 5), (dict(d=136), 5), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.inf), 1),
    (dict(scale=math.nan), 1), (dict(n_seq=0), 1), (dict(n_seq=1 << 20), 1), (dict(), 1),
])
def test_attention_refuses_before_any_device_call(libsc, change, status):
    assert attn(libsc, **change) == status
    assert len(libsc.sc_last_error()) > 0


def rope(L, tokens=4, hq=2, hk=2, d=64, rot=64, axes=1, eps=1e-6, amp=1.0, dtype=1, flags=0):
    return L.sc_qk_norm_rope_fwd(None, None, None, None, None, None, None, 1, axes, None, tokens, hq, hk, d, rot, eps,
                                 amp, dtype, flags, None)


@pytest.mark.parametrize("change,status", [
    (dict(flags=2), 1), (dict(dtype=7), 1), (dict(tokens=-1), 1), (dict(hq=-1), 1), (dict(d=12), 5), (dict(d=264), 5),
    (dict(rot=63), 1), (dict(rot=66), 1), (dict(rot=-2), 1), (dict(axes=0), 1), (dict(axes=3), 1), (dict(axes=5), 1),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(amp=math.inf), 1), (dict(), 1), (dict(rot=0), 1),
    (dict(tokens=0), 0), (dict(hq=0, hk=0), 0),
])
def test_rotation_refuses_before_any_device_call(libsc, change, status):
    assert rope(libsc, **change) == status


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 2, 64), dtype=torch.float16)
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.sc_attn_fwd(x, x, x, off)
    with pytest.raises(ValueError, match="CUDA tensor"):
        binding.sc_qk_norm_rope_fwd(x, x)
    with pytest.raises(ValueError, match="pass q"):
        binding.sc_qk_norm_rope_fwd(None, None)


def test_view_struct_matches_the_header():
    assert ctypes.sizeof(binding._Heads) == 24


def test_frequencies():
    f, amp = binding.rope_frequencies(64)
    assert f.dtype == torch.float32 and f.shape == (32,) and amp == 1.0
    want = [10000.0 ** (-i / 32) for i in range(32)]
    assert all(abs(float(a) - b) <= 1e-7 * b for a, b in zip(f, want))
    f3, _ = binding.rope_frequencies(60, axes=3)
    assert torch.equal(f3[:10], f3[10:20]) and torch.equal(f3[:10], f3[20:])
    lin, _ = binding.rope_frequencies(64, scaling="linear", factor=4.0)
    assert torch.allclose(lin * 4, f)
    base, _ = binding.rope_frequencies(64, scaling="base", factor=4.0)
    assert abs(float(base[0]) - 1) < 1e-7 and abs(float(base[-1]) * 4 / float(f[-1]) - 1) < 1e-5
    parts, amp = binding.rope_frequencies(64, scaling="parts", factor=8.0, original=4096)
    assert abs(amp - (1 + 0.1 * math.log(8.0))) < 1e-12
    assert float(parts[0]) == float(f[0])  # 650 turns over the original length: kept
    assert abs(float(parts[-1]) * 8 / float(f[-1]) - 1) < 1e-6  # under one turn: divided
    ratio = parts / f
    assert bool((ratio[1:] <= ratio[:-1] + 1e-7).all())
    for bad in (dict(rot_dim=63), dict(rot_dim=64, axes=3), dict(rot_dim=64, factor=0.5),
                dict(rot_dim=64, scaling="other")):
        with pytest.raises(ValueError):
            binding.rope_frequencies(**bad)
