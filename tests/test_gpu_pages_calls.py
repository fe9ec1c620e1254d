"""Page lists on the GPU: how calls treat what the caller passes."""
import numpy as np
import pytest

from test_gpu_pages import Pool

pytestmark = pytest.mark.gpu


def test_compaction_leaves_the_callers_dict_alone(tsv):
    """Results without a status of their own: the returned dict has one, the passed one is as it was."""
    p = Pool(tsv, np.random.default_rng(1), 300, [20, 7, 30], 40)
    first = tsv.pages_compact(p.pool, [p.d_table], [p.d_pages])
    want = {k: v.clone() for k, v in first.items() if k not in ("tables", "status")}
    out = {k: v for k, v in first.items() if k != "status"}
    names = set(out)
    got = tsv.pages_compact(p.pool, [p.d_table], [p.d_pages], out=out)
    assert set(out) == names and got["status"].tolist() == [0]
    for k, v in want.items():
        assert got[k] is out[k]
        m = int(got["moved"]) if k.startswith("move_") else None  # (entries behind the moves are not written)
        assert (got[k][:m] == v[:m]).all()
