"""The 8-bit product on its other paths: tables of one row."""
import numpy as np
import pytest
import torch

import embedding_lookup_tied_gb300 as lhs
from test_i8_product import make_rows, ref_logits, same, table_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [2, 30])
@pytest.mark.parametrize("k", [16, 63, 100, 897])
def test_table_of_one_row(m, k):
    # one row of k codes in a buffer that is as wide as a longer table's rows: any number of rows of
    # it is a table, so one is
    rng = np.random.default_rng([m, k])
    wb, ws = make_rows(rng, 5, k)
    ab, as_ = make_rows(rng, m, k)
    codes, scales = torch.from_numpy(wb).cuda(), torch.from_numpy(ws).cuda()
    tok = table_of(ab, as_, k)
    for rows in (2, 1):
        tab = lhs.lhs_i8_init(codes[:rows, :k], scales[:rows], k)
        out, err = lhs.lhs_i8_matmul(tok, tab)
        assert int(err.item()) == 0
        assert same(out, ref_logits(ab[:, :k], as_, wb[:rows, :k], ws[:rows], torch.float32)), rows
    t, _ = lhs.lhs_i8_quantize(torch.from_numpy(wb[:1, :k].astype(np.float32)).cuda())
    again = lhs.lhs_i8_init(t.codes, t.scales, k)
    assert lhs.lhs_i8_matmul(tok, again)[0].shape == (m, 1)
