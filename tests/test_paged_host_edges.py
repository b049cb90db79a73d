"""The paged cache without a GPU: the ends of the E4M3 format's range and the
Python layer's checks of its arguments."""

import numpy as np
import pytest

import oracle as O
from oracle import paged as OP


# ---- the oracle

@pytest.mark.parametrize("amax,code", [
    (255 * 2.0 ** 120, 0x77),  # BF16's largest: 240 * 2^120, since 256 * 2^120 is not finite
    (248 * 2.0 ** 120, 0x77),
    (247 * 2.0 ** 120, 0x77),
    (232 * 2.0 ** 120, 0x76),  # half way between 224 and 240: even
    (224 * 2.0 ** 120, 0x7E),  # 448 * 2^119
    (2.0 ** 127, 0x78),        # 256 * 2^119
])
def test_codes_stand_for_finite_values(amax, code):
    bits = np.zeros(128, dtype=np.uint16)
    bits[7] = int(np.array([amax], dtype=np.float32).view(np.uint32)[0]) >> 16
    bits[9] = bits[7] | 0x8000
    codes, byte = OP.quantise_row(bits)
    assert codes[7] == code and codes[9] == code | 128 and byte == (247 if code < 0x7E and amax > 2.0 ** 127 else 246)
    back = OP.dequantise(codes[None], np.array([byte]))[0]
    ref = O.decode_bf16(bits)
    assert np.all(np.abs(back) <= 255 * 2.0 ** 120)
    assert np.all(np.abs(back - ref) <= 2.0 ** -4 * np.abs(ref))


# ---- the Python layer

FIELDS = dict(kind=0, pages=10, H=2, page_size=64, D=128, seqs=3, table_width=4, table_stride=4, rows=7, max_new=7,
              Hq=4, causal=1, window=0, scale=0.1, at=512, ah=128, bt=512, bh=128)


@pytest.mark.parametrize("name", [n for n in FIELDS if n not in ("scale",)])
@pytest.mark.parametrize("value", [2 ** 63, -2 ** 63 - 1, 2 ** 64 + 16])
def test_numbers_that_the_structure_cannot_hold_are_refused(name, value):
    """ctypes would take them modulo 2^32 (2^64)."""
    from block_sparse_routed_gb300 import paged

    with pytest.raises(ValueError, match="range"):
        paged._params(*dict(FIELDS, **{name: value}).values())


@pytest.mark.parametrize("name", [n for n in FIELDS if n not in ("scale", "table_stride", "at", "ah", "bt", "bh")])
def test_numbers_past_32_bits_are_refused_where_the_structure_has_32(name):
    from block_sparse_routed_gb300 import paged

    for value in (2 ** 31, 2 ** 32 + 16, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="range"):
            paged._params(*dict(FIELDS, **{name: value}).values())
    p, _ = paged._params(*dict(FIELDS, at=2 ** 40, table_stride=2 ** 33).values())
    assert p.a_token_stride == 2 ** 40 and p.table_stride == 2 ** 33


def test_an_output_of_another_shape_is_refused():
    """As many elements in another order are not the output."""
    torch = pytest.importorskip("torch")
    from block_sparse_routed_gb300 import paged

    f32 = torch.float32
    for shape in ((3, 4), (1, 3, 4)):
        t = torch.zeros(shape)
        assert paged._given(t, "lse", (3, 4), f32, -1) is t
    for t in (torch.zeros(4, 3), torch.zeros(12), torch.zeros(3, 1, 4), torch.zeros(4, 3).t(), torch.zeros(2, 3, 4),
              torch.zeros(3, 4, dtype=torch.float64), torch.zeros(6, 4)[::2]):
        with pytest.raises(ValueError, match="lse"):
            paged._given(t, "lse", (3, 4), f32, -1)
