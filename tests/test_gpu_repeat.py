"""Causal calls repeated: the same inputs give the same bits every time.

Forward and gradient on the tensor cores at the tile layouts that overlap a chunk's products with the rows' epilogues
and denominators of the one before: one and two buffers of output sums, with and without cos/sin weights."""
import pytest
import torch

import gpu_helpers as H
from efficient_transformer_gb300 import build as la_build
from efficient_transformer_gb300 import inputs as gen
from efficient_transformer_gb300 import la

pytestmark = pytest.mark.gpu

CASES = [
    # B, Hq, Hkv, N, D, phi, weights
    (2, 16, 16, 8192, 128, "relu", True),    # one buffer of output sums, masked rows
    (2, 16, 8, 4096, 128, "elu+1", True),    # one buffer
    (2, 16, 16, 8192, 128, "relu", False),
    (2, 16, 8, 8192, 128, "elu+1", False),
    (2, 16, 4, 4096, 128, "elu+1", True),    # two buffers
    (4, 16, 16, 4096, 64, "relu", True),
    (4, 16, 8, 4096, 64, "elu+1", False),
]


@pytest.fixture(scope="module", autouse=True)
def built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    la_build.build()
    la.load()


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_repeated_calls_give_the_same_bits(case):
    B, Hq, Hkv, N, D, phi, weights = case
    w = gen.Workload(f"repeat_b{B}_hq{Hq}_hkv{Hkv}_n{N}_d{D}_{phi}", B, Hq, Hkv, N, D, "bf16", True, phi, scale=0.5,
                     weights=weights)
    dev = H.to_dev(gen.make_inputs(w, seed=17))
    first = [t.clone() for t in H.run_gpu(w, dev, from_fwd=True)]
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")   # calls with other bits
    for _ in range(200):
        got = H.run_gpu(w, dev, from_fwd=True)
        wrong += torch.stack([(a != b).any() for a, b in zip(got, first)]).any()
    assert wrong.item() == 0, f"{wrong.item()} of 200 calls differ from the first"
