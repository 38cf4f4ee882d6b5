"""Packed attention gives the same bits in every run, also where the batch's
last round of items is cut into parts: which of several equally long tiles is
cut must follow from the batch, not from the order in which the planning warps
arrive. A cut tile is summed up in another order, so its bits show it.

Each case has tiles of equal length on both sides of the cut (128 / G tokens,
two of them per tile; 152 SMs, an item per KV head). Between runs the caches
are flushed, other kernels' code goes through the instruction cache, or work
runs beside the call, which moves the warps against one another."""
import pytest

from tests import _packed as K

pytestmark = pytest.mark.gpu

L = K.Layout
LLAMA = L(32, 8, 128, 4)

CASES = {
    # 20 equal tiles of 8 KV heads: one of them is cut
    "equal_tiles_over_one_round": (LLAMA, [64] * 20, [0] * 20, 640),
    # two lengths in turn, the longer ones whole; 40 tiles: the second round's last two are cut
    "two_lengths_over_two_rounds": (LLAMA, [60] * 40, [300 * (i % 2) + 500 for i in range(40)], 0),
    # unlike prompts behind a long text, not shared
    "unlike_prompts_behind_a_text": (LLAMA, [1 + (97 * i) % 340 for i in range(9)] + [64] * 8, [0] * 17, 2048),
    # one long prompt: its tiles belong to eight warps, four of them share a number of blocks
    "one_prompt_over_one_round": (L(4, 4, 64, 1), [256 * 40], [0], 0),
}


@pytest.mark.parametrize("name", list(CASES))
def test_every_run_gives_the_same_bits(gpu_lib, name):
    import torch
    lay, new, cached, prefix = CASES[name]
    b = K.Batch(lay, new, cached, prefix=prefix, seed=21)
    d = K.OnDevice(gpu_lib, b)
    first = d.run().clone()
    assert d.status() == 0
    flush = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")
    x = torch.randn(1024, 1024, device="cuda")
    side = torch.cuda.Stream()
    different = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(150):
        if i % 3 == 1:
            flush.fill_(i)
        if i % 4 == 2:
            torch.sort(x.view(-1)[:4096 + i])
        if i % 5 == 3:
            with torch.cuda.stream(side):
                x @ x
        d.out.fill_(7.0)
        different += (d.run() != first).any()
    torch.cuda.synchronize()
    assert different.item() == 0, f"{different.item()} of 150 runs differ"
