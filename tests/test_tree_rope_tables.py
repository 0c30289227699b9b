"""A rotation table that the caller fills: any frequencies, in 2^-64 turns a
position, as the documentation says."""

import math

import numpy as np
import pytest
import torch

import layer_gram_embedding_gb300 as ple
import tree_reference as ref
from test_tree_ops import U, check_rows, dev, host, rows

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def index_ramp(R, base, factor, trained, fast, slow):
    """Interpolation by parts with the ramp over the pairs' indices, between those of `fast` and `slow` turns."""
    def pair(turns):
        return R * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

    low, high = math.floor(pair(fast)), math.ceil(pair(slow))
    i = np.arange(R // 2)
    keep = 1 - np.clip((i - low) / (high - low), 0, 1)
    w = base ** (-2.0 * i / R)
    return keep * w + (1 - keep) * w / factor


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("kind", ["index ramp", "any"])
def test_a_table_of_the_callers_own(kind, interleaved, dtype):
    rng = np.random.default_rng(91)
    R = D = 128
    w = index_ramp(R, 1e6, 4.0, 32768.0, 32.0, 1.0) if kind == "index ramp" \
        else rng.uniform(0.0, 3.0, R // 2)
    rope = (torch.from_numpy(w).double() / (2 * math.pi) * 2.0 ** 64).long().cuda()
    q, k = rows(rng, (50, 3, D), dtype, 2.0), rows(rng, (50, 1, D), dtype, 2.0)
    positions = rng.integers(0, 131072, 50).astype(np.int32)
    got = ple.ple_qk_norm_rope(q, k, None, dev(positions), rope, interleaved=interleaved)
    for x, y in zip((q, k), got):
        want, size = ref.norm_rope(host(x), None, positions, w, 0.0, interleaved, 1.0)
        check_rows(y, want, size, U[dtype], kind)


def test_the_two_ramps_are_not_one():
    # the figure in the documentation: a pair of about 5.7 turns
    w = ref.inverse_frequencies(128, 1e6, "plain")
    turns = 32768.0 * w / (2 * math.pi)
    i = int(np.argmin(np.abs(turns - 5.7)))
    by_index = index_ramp(128, 1e6, 4.0, 32768.0, 32.0, 1.0)[i] / w[i]
    by_turns = ref.inverse_frequencies(128, 1e6, "parts", 4.0, 32768.0)[i] / w[i]

    def keep(x):
        return (x - 0.25) / 0.75

    assert abs(keep(by_turns) - 0.15) < 0.03 and abs(keep(by_index) - 0.5) < 0.05
