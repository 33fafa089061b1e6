"""Host side of the new-token operators where numbers are at the end of their range: score scales and rotary steps."""
import ctypes

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
