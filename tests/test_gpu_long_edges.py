"""The operators for long contexts at the ends of their inputs' ranges, on the GPU: scores
past fp32, bounds never written, table entries that name no block, requests longer than what
is held in shared memory, caches of several layers."""
import numpy as np
import pytest
import torch

import long_reference as R
from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu


class Bounds:
    """Requests of these lengths (new tokens: 1 each) with codes and scales and no keys."""

    def __init__(self, lens, n_kv, d, seed, block=16):
        rng = np.random.default_rng(seed)
        self.lens, self.n_kv, self.d, self.block = list(lens), n_kv, d, block
        self.tokens = len(lens)
        self.starts = np.arange(len(lens) + 1)
        held = [-(-n // block) for n in lens]
        self.blocks = sum(held) + 2
        ids = rng.permutation(self.blocks)
        self.tables = np.full((len(lens), max(held)), -1, np.int32)
        at = 0
        for s, n in enumerate(held):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.codes = torch.from_numpy(
            rng.integers(-127, 128, (self.blocks, n_kv, 2, d))).to(torch.int8).cuda()
        self.scales = torch.ones(self.blocks, n_kv, device="cuda")

    def choose(self, q, n_sel, sinks, recent, guard=3):
        """(chosen, the rows before and behind them)."""
        i32 = dict(dtype=torch.int32, device="cuda")
        rows = torch.full((self.tokens + 2 * guard, self.n_kv, n_sel), -9, **i32)
        out = rows[guard:guard + self.tokens]
        ops.select_blocks(q, self.codes, self.scales, torch.from_numpy(self.tables).cuda(),
                          torch.tensor(self.lens, **i32), torch.tensor(self.starts, **i32),
                          num_selected=n_sel, num_sinks=sinks, num_recent=recent,
                          block_size=self.block, max_seq_len=max(self.lens), out=out)
        ops.check_device_errors()
        return out.cpu().numpy(), torch.cat([rows[:guard], rows[guard + self.tokens:]])


@pytest.mark.parametrize("scores", ["nan scales", "past fp32 by no scale"])
@pytest.mark.parametrize("lens", [[640, 300, 4096], [16000, 640], [40000, 17000, 300]])
def test_scores_of_no_number_stay_in_their_row(lens, scores):
    """Blocks whose bounds hold anything: as many as asked for are chosen, no more."""
    b = Bounds(lens, 2, 128, seed=1)
    q = torch.ones(len(lens), 16, 128, dtype=torch.bfloat16, device="cuda")
    if scores == "nan scales":
        b.scales.fill_(float("nan"))
    else:
        q.fill_(2.0 ** 115)  # (each sum is past fp32 and then multiplied by a scale of 0)
        b.codes.fill_(127)
        b.scales.zero_()
    for n_sel, sinks, recent in ((5, 1, 2), (3, 1, 2), (16, 0, 1)):
        got, guard = b.choose(q, n_sel, sinks, recent)
        assert (guard == -9).all()
        assert (np.diff(got, axis=-1) > 0).all() and (got >= 0).all()
        assert (got[..., -1] < -(-np.array(lens)[:, None] // 16)).all()
