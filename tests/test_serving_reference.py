"""CPU checks of the serving operators: the 4-bit format's own properties, and the binding's refusals (made before
anything reaches the library)."""
import numpy as np
import pytest
import torch

import kv_cache_retention_gb300 as kv
import serving_reference as ref


def test_scale_bytes_are_the_top_of_fp16():
    bits = (np.arange(227, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    assert np.array_equal(bits, ref.LADDER)
    assert np.all(np.diff(ref.LADDER) > 0) and ref.LADDER[-1] == 10240 and np.isnan(ref.scale_value(255))


def test_every_stored_value_is_exact_in_bf16_and_fp16():
    vals = (ref.MAGS[:, None] * ref.LADDER[None]).ravel()
    t = torch.from_numpy(vals)
    assert torch.equal(t.to(torch.bfloat16).double(), t) and torch.equal(t.to(torch.float16).double(), t)


def test_quantise_known_groups():
    x = np.zeros((4, 16))
    x[0, :8] = [6, -6, 0.25, 0.75, 2.5, 3.5, 5, -0.25]     # scale 1; ties go to the even code
    x[1, 0] = 61440
    x[2, 3] = np.nan
    x[3, 3] = 61441
    codes, scales = ref.quantise(x)
    assert scales[:, 0].tolist() == [15 << 3, 226, 255, 255]
    assert ref.dequantise(codes, scales)[0, :8].tolist() == [6, -6, 0, 1, 2, 4, 4, 0]
    assert ref.dequantise(codes, scales)[1, 0] == 61440
    assert np.isnan(ref.dequantise(codes, scales)[2:]).all() and not codes[2:].any()


def test_stored_values_are_within_one_scale():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * 10.0 ** rng.uniform(-6, 4, (200, 1))
    codes, scales = ref.quantise(x)
    s = np.repeat(ref.scale_value(scales), 16, -1)
    assert np.all(np.abs(ref.dequantise(codes, scales) - x) <= s)


class _Fake:
    """A context object without a device, for checks that come before the library."""

    def __new__(cls):
        c = object.__new__(kv.Context)
        c.device, c.handle = 0, None
        return c


def test_cpu_tensors_are_refused():
    c = _Fake()
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        c.prompt_attention(q, q, q, torch.zeros(2, dtype=torch.int32), q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        c.kv4_store(q, q, None, None, None, None, None)
    with pytest.raises(ValueError, match="CUDA tensor"):
        i = torch.zeros(1, dtype=torch.int32)
        c.plan_slots(i, i, i, 16, 1, torch.zeros((1, 1), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), i, i,
                     torch.zeros(2, dtype=torch.int32))


def test_row_spacing():
    """Rows at an even spacing, an expanded token axis (spacing 0, which the library refuses) among them."""
    bf = torch.bfloat16
    x = torch.zeros((6, 4, 64), dtype=bf)
    at = lambda t, lead: kv._rows(t, lead, bf, -1, "x")[1]  # noqa: E731
    assert at(x, 1) == 256 and at(x[:, 1:3], 1) == 256 and at(x[::2], 1) == 512 and at(x[:1, :2], 1) in (128, 256)
    assert at(x[:1].expand(5, 4, 64), 1) == 0
    assert at(x[:1].unsqueeze(1).expand(5, 3, 4, 64), 2) == 0
    assert at(x.view(3, 2, 4, 64)[:, :, :2], 2) == 256
    for bad in (x[:3].unsqueeze(1).expand(3, 2, 4, 64), x[:2].unsqueeze(0).expand(3, 2, 4, 64)):
        with pytest.raises(ValueError, match="evenly spaced"):
            at(bad, 2)


def test_null_context_is_refused():
    z = [None] * 32
    assert kv.kvsel_plan_slots(None, None, None, 1, 16, 1, None, 0, None, 1, None, None, None, 0, None, 0, None,
                               None) == kv.ERR_INVALID_ARG
    assert kv.kvsel_kv4_store(None, None, None, kv.BF16, 128, 128, 1, 1, 128, *z[:5], 1, 16, None) == kv.ERR_INVALID_ARG
    assert kv.kvsel_kv4_load(None, *z[:4], 1, 16, None, 1, 1, 128, None, None, 128, 128, None) == kv.ERR_INVALID_ARG
    assert kv.kvsel_kv4_attention(None, None, 128, 1, 1, 1, 1, 128, *z[:4], 1, 16, *z[:3], 1, -1, 1.0, None, None,
                                  None) == kv.ERR_INVALID_ARG
    assert kv.kvsel_prompt_attention(None, None, None, None, 128, 128, 128, None, 1, 1, 1, 1, 128, 1.0, None, None,
                                     None) == kv.ERR_INVALID_ARG
