"""Host side of the new-token operators where numbers are at the end of their range: score scales and rotary steps."""
import ctypes
import math
from decimal import Decimal, getcontext

import pytest

from compressed_kv_cache_quant_gb300 import _abi, kvq
from compressed_kv_cache_quant_gb300.build import build

pytestmark = pytest.mark.cpu
by = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    build()
    return kvq.lib()


@pytest.mark.parametrize("scale,softcap", [(3e38, 0.0), (2.4e38, 0.0), (3e38, 1e38)])
def test_scale_beyond_fp32_in_log2_units_is_refused(lib, scale, softcap):
    """Scores are kept in log2 units: a scale whose product with log2(e) = 1.44 is no fp32 number would make every score
    infinite or NaN.  The largest scale below that is taken."""
    L = kvq.make_layout(8, 2, 16)
    pool = _abi.Pool(num_blocks=16, max_seqs=4, t_cap=0, k16=256, v16=256)
    seqs = _abi.Seqs(256, 256, 0, 8, 100, 0)   # a batch of none: accepted calls launch nothing
    for bad in (True, False):
        mod = _abi.AttnModStruct(scale if bad else 2.3e38, softcap)
        got = (lib.kv_decode_attn(by(L), by(pool), by(seqs), 256, by(mod), 256, None, 256, 1 << 30, None),
               lib.kv_chunk_attn(by(L), by(pool), by(seqs), 256, 256, 4, 2, by(mod), 256, None, 256, 1 << 30, None))
        assert got == ((_abi.KVQ_ERR_INVALID_ARG,) * 2 if bad else (0, 0)), kvq._abi.last_error()


def turns_of(rot, kind, original, base, factor, low, high):
    """Turns per position of every pair, to 60 digits."""
    getcontext().prec = 60
    # pi = 16 atan(1/5) - 4 atan(1/239)
    atan = lambda n: sum((-1) ** k / (Decimal(2 * k + 1) * Decimal(n) ** (2 * k + 1)) for k in range(45))  # noqa: E731
    pi = 16 * atan(5) - 4 * atan(239)
    b, x = Decimal(base), Decimal(factor)
    if kind == "ntk":
        b = b * (Decimal(rot) / (rot - 2) * x.ln()).exp()
    out = []
    for i in range(rot // 2):
        f = (-Decimal(2 * i) / rot * b.ln()).exp()
        keep = Decimal(0 if kind == "linear" else 1)
        if kind == "yarn":
            at = [rot * (Decimal(original) / (Decimal(n) * 2 * pi)).ln() / (2 * b.ln()) for n in (low, high)]
            lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
            keep = 1 - min(max(Decimal(i - lo) / max(Decimal(hi - lo), Decimal("0.001")), Decimal(0)), Decimal(1))
        if kind == "knees":
            keep = min(max((original * f / (2 * pi) - Decimal(low)) / (Decimal(high) - Decimal(low)), Decimal(0)), Decimal(1))
        out.append((f * keep + f / x * (1 - keep)) / (2 * pi) if kind in ("linear", "yarn", "knees") else f / (2 * pi))
    return out


@pytest.mark.parametrize("rot", [16, 96, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1000000.0])
@pytest.mark.parametrize("kind,factor,original,low,high", [("plain", 1.0, 0, 0.0, 0.0), ("linear", 4.0, 0, 0.0, 0.0),
                                                           ("ntk", 8.0, 0, 0.0, 0.0), ("yarn", 4.0, 32768, 32.0, 1.0),
                                                           ("knees", 8.0, 8192, 1.0, 4.0)])
def test_rope_angles_at_far_positions(lib, rot, base, kind, factor, original, low, high):
    """The wrapped product of a position and a step against the angle itself, both in turns.  A step is within 2^-48 of itself
    (the power's exponent is rounded, 2^-53 of it times ln(base) < 14; the power, the division and the ramp add a few
    2^-53) and 2^-63 turns (the fraction's last two units)."""
    r = _abi.Rope(rot, 0, _abi.ROPE_SCALINGS[kind], original, base, factor, low, high)
    steps, m = (ctypes.c_uint64 * 64)(), ctypes.c_float(0)
    assert lib.kvq_rope_steps(by(r), steps, by(m)) == 0
    for i, f in enumerate(turns_of(rot, kind, original, base, factor, low, high)):
        off = f * Decimal(2) ** -48 + Decimal(2) ** -63
        for p in (1, 4097, 131071, 10 ** 6 + 3, 2 ** 31 - 1, -77777, -2 ** 31):
            got = Decimal(p * steps[i] % 2 ** 64) / Decimal(2) ** 64
            gap = abs(got - p * f % 1) % 1
            assert min(gap, 1 - gap) <= abs(p) * off, (i, p)


def test_max_len_beyond_2_30_is_refused(lib):
    """Positions, pages and tiles are counted in 32 bits with sums of two of them: the attention of new tokens takes up to 2^30
    tokens a sequence (512 GB of an fp16 layer with one kv head)."""
    L = kvq.make_layout(8, 2, 16)
    pool = _abi.Pool(num_blocks=16, max_seqs=4, t_cap=0, k16=256, v16=256)
    for max_len, want in ((2 ** 30, 0), (2 ** 30 + 1, _abi.KVQ_ERR_UNSUPPORTED), (2 ** 31 - 1, _abi.KVQ_ERR_UNSUPPORTED)):
        seqs = _abi.Seqs(256, 256, 0, 2 ** 27, max_len, 0)   # a batch of none
        assert lib.kv_decode_attn(by(L), by(pool), by(seqs), 256, None, 256, None, 256, 1 << 40, None) == want
        assert lib.kv_chunk_attn(by(L), by(pool), by(seqs), 256, 256, 4, 2, None, 256, None, 256, 1 << 40, None) == want
        seqs.batch = 1
        assert (lib.kv_decode_attn_ws(by(L), by(seqs)) == 0) == (want != 0)
        assert (lib.kv_chunk_attn_ws(by(L), by(seqs), 4, 2) == 0) == (want != 0)
