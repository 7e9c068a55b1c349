"""The numpy definition of the 4-bit cache pinned by facts that do not come
from it: representability, the quantiser's error, the layout's bijection."""
import numpy as np
import pytest
import torch

import kv4_reference as ref


def test_every_stored_value_is_a_bf16_and_an_fp16_number():
    x = np.unique(np.concatenate([s * np.arange(-15, 16) for s in ref.scales()]))
    t = torch.from_numpy(x)
    assert torch.equal(t.to(torch.bfloat16).double(), t)
    assert torch.equal(t.to(torch.float16).double(), t)
    assert ref.scales()[-1] == 3840 and ref.scales()[1] == 2.0**-17
    fp16 = torch.arange(0xD8, dtype=torch.int16).mul(128).view(torch.float16).double().numpy()
    assert np.array_equal(fp16, ref.scales())


@pytest.mark.parametrize("scale", [1e-3, 1.0, 300.0])
def test_quantisation_error_is_half_a_step_and_what_the_scale_rounding_clips(scale):
    # the step is at most 1/16 off (3 bits of mantissa), so the 15 steps miss
    # up to 15/16 of a step of the span; the zero point moves it by another
    # half: an element is off by at most 0.5 + 15/16 + 0.5 steps, and steps
    # are at most 17/16 of span / 15
    rng = np.random.default_rng(5)
    x = torch.from_numpy(rng.standard_normal((400, 128)) * scale).to(torch.bfloat16).double().numpy()
    g = x.reshape(-1, 4, 32)
    span = np.maximum(g.max(-1), 0) - np.minimum(g.min(-1), 0)
    err = np.abs(ref.stored(x) - x).reshape(g.shape)
    assert (err <= (2 * 17 / 16 * span / 15)[..., None] + 2.0**-17).all()
    # and on average less than half a step
    assert np.sqrt((err**2).mean()) < 0.5 * (span / 15).mean()


def test_zero_is_stored_exactly_and_tiny_rows_do_not_fail():
    x = np.zeros((3, 128))
    x[1, ::3] = 5.5
    x[2] = 1e-30
    assert (ref.stored(x)[x == 0] == 0).all()
    assert np.abs(ref.stored(x)[2]).max() <= 2.0**-17


def test_saturation_and_nan():
    x = np.full((1, 128), 1.0)
    x[0, :4] = [np.inf, -np.inf, np.nan, 1e30]
    y = ref.stored(x)[0]
    assert y[2] == 0 and y[0] == y[3] and abs(y[0] - ref.TOP) <= 3840 and abs(y[1] + ref.TOP) <= 3840
    assert np.abs(y[4:]).max() <= 3840  # the rest of that group; the other groups are as ever
    assert np.abs(y[32:] - 1).max() <= 17 / 16 / 15


def test_pack_and_unpack_are_inverse_and_use_every_bit():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 2, 128, 128))
    t = ref.pack(k, v)
    k2, v2 = ref.unpack(t)
    assert np.array_equal(k2, ref.stored(k)) and np.array_equal(v2, ref.stored(v))
    for is_v in (False, True):
        byte, shift = ref._places(is_v)
        assert len({(b, s) for b, s in zip(byte.reshape(-1), shift.reshape(-1))}) == 64 * 128 and byte.max() == 4095


def test_evict_keeps_the_heaviest_the_last_and_the_lower_of_equals():
    acc = np.array([1.0, 3.0, 2.0, 3.0, np.nan, 2.0, 0.0, -1.0])
    assert list(ref.evict(acc, 8, 4, 1)) == [1, 2, 3, 7]
    assert list(ref.evict(acc, 8, 7, 0)) == [0, 1, 2, 3, 5, 6, 7]
    assert list(ref.evict(acc, 8, 8, 3)) == list(range(8))
    assert list(ref.evict(acc, 8, 2, 2)) == [6, 7]
