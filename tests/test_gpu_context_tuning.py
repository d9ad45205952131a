"""The decode inside the forms for long and shared contexts follows the tuning's CTA counts and tiers."""
import numpy as np
import pytest
import torch

import paged_kv_gqa_split_gb300 as pkg
from paged_kv_gqa_split_gb300 import _lib
from paged_kv_gqa_split_gb300.build import build
import test_gpu_blocks as blocks_of
import test_gpu_shared as shared
import test_gpu_weights as weights

pytestmark = pytest.mark.gpu

TUNINGS = [dict(num_ctas=1), dict(num_ctas=7), dict(num_ctas=150, tier2_ctas=-1), dict(tier2_ctas=-1), dict(tier2_ctas=40),
           dict(num_ctas=13, tier2_ctas=5, tier2_permille=500, tier2_min_units=3), dict(tier2_permille=700), dict(tier2_min_units=1),
           dict(min_units_per_cta=200), dict(num_ctas=1536)]


@pytest.fixture(scope="module", autouse=True)
def _library(cuda_device):
    build()
    _lib.load()


@pytest.fixture(autouse=True)
def _defaults():
    yield
    _lib.gqa_paged_decode_set_tuning()


def tuned(tuning):
    assert _lib.gqa_paged_decode_set_tuning(**tuning) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[3000, 0, 17, 900, 1], [5] * 100, [20000]])
@pytest.mark.parametrize("tuning", TUNINGS, ids=str)
def test_weights_follow_the_tuning(tuning, lens, fp8):
    """The plain decode under the same tuning cuts the same pieces: the same bits."""
    args = weights.make(lens, max(lens), fp8, sum(lens))
    tuned(tuning)
    got = pkg.run_weighted(*args, decay=0.5)
    weights.check(args, 0.5, got)
    out, lse = (pkg.run_fp8 if fp8 else pkg.run)(*args[:5])
    assert torch.equal(out, got[0]) and torch.equal(lse, got[1])


@pytest.mark.parametrize("rows", [1, 2])
@pytest.mark.parametrize("tuning", TUNINGS, ids=str)
def test_chosen_blocks_follow_the_tuning(tuning, rows):
    """Every block chosen: the selected-token decode of all tokens under the same tuning gives the same bits where a row's
    places are the same in both, which they are for lengths of whole blocks."""
    lens, page = [640, 640, 640], 16
    w = blocks_of.make(lens, page, 3, rows)
    w["row_lens"] = blocks_of.i32([640] * (3 * rows))
    pkg.block_bounds(w["k"], w["bounds"], w["table"], w["lens"])
    tuned(tuning)
    chosen = blocks_of.select(w, 40)
    out, lse = blocks_of.attend(w, chosen)
    blocks_of.check(w, chosen, out, lse)
    tokens = torch.arange(640, dtype=torch.int32).cuda().expand(3 * rows, 640).contiguous()
    want, want_lse = pkg.sparse_run(w["q"], w["k"], w["v"], tokens, w["table"], w["req"])
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", [([1000], [20], [300, 0, 7]), ([], [], [2000, 40]), ([0, 130], [3, 70], [40])], ids=str)
@pytest.mark.parametrize("tuning", TUNINGS, ids=str)
def test_shared_prefixes_under_a_tuning(tuning, case, fp8):
    prefixes, members, own = case
    args = shared.make(prefixes, members, 2, own, fp8, seed=sum(own))
    tuned(tuning)
    shared.check(args, *pkg.shared_run(*args))


def test_a_workspace_is_what_the_tuning_asks_for():
    args = shared.make([300], [5], 0, [100], seed=1)
    small = _lib.load().gqa_shared_paged_decode_ws_size(5, 1, 0)
    tuned(dict(num_ctas=1536))
    large = _lib.load().gqa_shared_paged_decode_ws_size(5, 1, 0)
    assert large > small
    with pytest.raises(pkg.GqaError):
        pkg.shared_run(*args, workspace=torch.zeros(small, dtype=torch.uint8, device="cuda"))
    out, lse = pkg.shared_run(*args, workspace=torch.full((large,), 0xFF, dtype=torch.uint8, device="cuda"))
    shared.check(args, out, lse)
    assert np.isfinite(out.float().cpu().numpy()).all()
