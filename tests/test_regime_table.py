"""The shipped regime table: every row parses, and the short classes keep the tiles that
they had before the 128-row kernel's whole-warp issuer.  (A table profiled at 8 heads of
4,096 tokens alone took 36 us instead of 19 for 4 heads of 2,048 tokens at 64 x 64, and
241 instead of 159 for 24 spatial SVG heads of 8,000.)"""
import pytest

import block_sparse_attention_tsr_gb300 as tsr


@pytest.fixture(scope="module", autouse=True)
def _table():
    tsr.build()
    tsr.lib()
    tsr.tsr_regime_load(tsr.REGIME_TABLE)


@pytest.mark.parametrize("kind,bq,bk,N,density,want", [
    (tsr.UNIFORM, 64, 64, 2048, 0.2, (64, 2, 1, tsr.ORIENT_KEYS)),
    (tsr.UNIFORM, 64, 64, 8000, 0.35, (64, 2, 1, tsr.ORIENT_KEYS)),
    (tsr.UNIFORM, 64, 64, 1024, 0.5, (64, 2, 1, tsr.ORIENT_KEYS)),
    (tsr.UNIFORM, 64, 64, 4096, 0.8, (64, 2, 1, tsr.ORIENT_KEYS)),
    (tsr.UNIFORM, 32, 32, 2048, 0.5, (64, 2, 2, tsr.ORIENT_ROWS)),
    (tsr.KEYLIST, 64, 1, 2048, 0.05, (64, 2, 1, tsr.ORIENT_KEYS)),
    (tsr.KEYLIST, 64, 1, 4096, 0.28, (64, 2, 2, tsr.ORIENT_ROWS)),
    (tsr.SVG, 0, 0, 8000, 0.06, (64, 4, 1, tsr.ORIENT_ROWS)),
    (tsr.UNIFORM, 64, 64, 32760, 0.25, (64, 2, 1, tsr.ORIENT_KEYS)),
    (tsr.UNIFORM, 64, 64, 32760, 0.5, (64, 2, 2, tsr.ORIENT_ROWS)),
])
def test_rows(kind, bq, bk, N, density, want):
    r = tsr.tsr_regime_lookup(kind, bq, bk, N, density)
    assert (r["bn"], r["stages"], r["ctas_per_sm"], r["orient"]) == want and r["id"] >= 0
