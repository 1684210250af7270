"""The plain forms of perf/operators.py, and the package's own calls beside them, against the
integer oracle, where their outputs are whole rows moved as they are."""
import numpy as np
import pytest
import torch

from perf import operators
from tests.helpers import cuda_or_skip, to_np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("pages,seqs", [(160, 6), (2040, 96)])
def test_compaction_moves_every_page_that_changes_its_number(pages, seqs, own, monkeypatch):
    """Both forms, twice on one state as they are measured: table, counts, numbers and the
    whole pool, holes among it, equal the oracle's."""
    from oracle import paged as op
    cuda_or_skip()
    monkeypatch.setattr(operators, "own", own)
    case = dict(op="compact", seqs=seqs, pages=pages, live=0.6, layers=1, kv=1, page=16)
    state = operators.prepare(case, 7)
    refs, table, data = (state[n].cpu() for n in ("refs", "table", "data"))
    refs, table, data = refs.numpy().copy(), table.numpy().copy(), to_np(data)
    remap = op.compact(data, refs, table, state["lengths"].tolist())
    for _ in range(2):
        got = operators.run(state)
        for x, want in zip(got, (table, refs, remap, data)):
            np.testing.assert_array_equal(to_np(x), want)
    torch.cuda.synchronize()
