"""Refusals of the 4-bit cache, windowed attention and QK-norm entry points
that need no GPU, and the page arithmetic that the GPU tests compare with."""
import numpy as np
import pytest

from speculative_decoding_exact_gb300 import abi
from tests import kv4_util as u


def test_null_arguments_are_refused():
    L = abi.lib()
    assert L.spec_qk_norm_rope(None, None, 0, 0, None, None, None, None, 0) == abi.SPEC_ENULL
    assert L.spec_kv4_append(None, None, 0, None, None, 0, 0) == abi.SPEC_ENULL
    assert L.spec_kv4_read(None, None, 0, 0, 0, None, None, 0) == abi.SPEC_ENULL
    assert L.spec_attention_kv4(None, None, 0, None, 1, 0, 0, None) == abi.SPEC_ENULL
    assert L.spec_attention_window(None, None, 0, None, 1, 0, 0, None) == abi.SPEC_ENULL


def test_page_size_agrees_with_the_header():
    text = open(abi.HEADER).read()
    assert f"#define SPEC_KV4_PAGE_BYTES {abi.KV4_PAGE_BYTES}" in text


def test_every_scale_byte_stands_for_its_binary16_number():
    vals = u.scale_values()
    assert vals[0] == 0 and vals[1] == 2.0 ** -17 and vals[0x78] == 1.0 and vals[-1] == 10240
    assert np.all(np.diff(vals) > 0)


@pytest.mark.parametrize("seed", [0, 1])
def test_quantise_is_nearest_under_the_smallest_sufficient_scale(seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((64, 16)) * 10.0 ** rng.integers(-6, 5, (64, 1))).astype(np.float32)
    code, byte = u.quantise(x)
    vals = u.scale_values()
    val = u.code_values()[code] * vals[byte]
    top = np.abs(x).max(-1).astype(np.float64)
    for i in range(64):
        b = byte[i, 0]
        assert b == 0xE2 or 6 * vals[b] >= top[i]
        assert b == 0 or 6 * vals[b - 1] < top[i]
        grid = u.code_values() * vals[b]
        best = np.abs(x[i, :, None].astype(np.float64) - grid).min(-1)
        assert np.array_equal(np.abs(x[i].astype(np.float64) - val[i]), best)


def test_pages_round_trip():
    rng = np.random.default_rng(3)
    code = rng.integers(0, 16, (32, 3, 128)).astype(np.uint8)
    byte = rng.integers(0, 256, (32, 3, 8)).astype(np.uint8)
    pages = u.to_pages(code, byte)
    assert pages.shape == (2, 3, abi.KV4_PAGE_BYTES)
    # positions from the format's text, one by one
    for t, h, e in [(0, 0, 0), (5, 1, 37), (17, 2, 127), (31, 0, 64)]:
        pg, tt = pages[t // 16, h], t % 16
        b = pg[256 * (e // 32) + 16 * tt + (e % 32) // 2]
        assert (b >> 4 if e % 2 else b & 15) == code[t, h, e]
        assert pg[1024 + 8 * tt + e // 16] == byte[t, h, e // 16]
    val = u.from_pages(pages)
    want = u.code_values()[code] * u.scale_values()[np.minimum(byte, 0xE2)].repeat(16, -1)
    assert np.array_equal(val, want)
