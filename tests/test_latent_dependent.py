"""Kernels that may be on the GPU before the kernel ahead of them has ended: they see what it wrote."""
import glob
import os
import re

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "hybrid_linear_attention_decode_gb300", "csrc")


def test_dependent_kernels_make_no_non_coherent_loads():
    """A non-coherent load is defined for memory that nothing writes during the kernel's lifetime."""
    files = [f for f in sorted(glob.glob(os.path.join(CSRC, "*.cu"))) if "wait_for_previous()" in open(f).read()]
    assert len(files) >= 3
    for f in files + [os.path.join(CSRC, "kda_latent.cuh")]:
        code = re.sub(r"//[^\n]*", "", open(f).read())
        for word in (r"__ldg\b", r"\.nc\b", r"__restrict"):
            assert not re.search(word, code), (f, word)


# A narrow table: rows of 3 entries, so that one 32-byte sector holds entries of several rows
ROWS, WIDTH, PAGE, RANK, ROPE, H = 12, 3, 16, 128, 64, 8


class Step:
    """A pool operation, directly followed by decodes of two layers over all rows."""

    def __init__(self, op, seed):
        import hybrid_linear_attention_decode_gb300 as kda
        from tests.test_latent_gpu import _i32
        self.kda, self.op = kda, op
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.pt = kda.PageTable.empty(ROWS, WIDTH, 48, PAGE)
        pages = torch.randn(2, 48, PAGE, RANK + ROPE, generator=g, device="cuda").to(torch.bfloat16)
        self.cache = kda.LatentCache(pages, RANK)
        self.st = _i32([0])
        self.pws = torch.empty(kda.kda_pages_workspace_bytes(self.pt, ROWS), dtype=torch.uint8, device="cuda")
        self.dws = torch.empty(kda.kda_latent_decode_workspace_bytes(self.cache, H, ROWS, 1), dtype=torch.uint8, device="cuda")
        self.q = torch.randn(ROWS, H, RANK + ROPE, generator=g, device="cuda").to(torch.bfloat16)
        self.out = torch.empty(2, ROWS, H, RANK, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.empty(2, ROWS, H, device="cuda")
        self.cu = torch.arange(ROWS + 1, dtype=torch.int32, device="cuda")
        # rows 0..7 of 9 to 37 tokens, over pages that are then scattered by ending rows between them
        lens = [9 + 4 * i for i in range(8)]
        kda.kda_pages_reserve(self.pt, self.cache, _i32([8, 9]), _i32([40, 40]), self.pws, self.st)
        for i in range(8):
            kda.kda_pages_reserve(self.pt, self.cache, _i32([i, 10]), _i32([lens[i], min(48, 6 * (i + 1))]), self.pws, self.st)
        kda.kda_pages_truncate(self.pt, _i32([8, 9, 10]), _i32([0, 0, 0]), self.pws, self.st)
        torch.cuda.synchronize()
        assert int(self.st.item()) == 0
        self.args = {"compact": (), "fork": ([7, 3, 5, 1], [8, 9, 10, 11]), "truncate": ([0, 2, 4, 6], [0, 5, 16, 20]),
                     "reserve": ([0, 2, 4, 6, 8], [10, 18, 26, 34, 1])}[op]
        self.arrays = [_i32(x) for x in self.args]
        self.kept = [x.clone() for x in (self.pt.table, self.pt.lens, self.pt.refcount, pages)]

    def restore(self):
        for have, kept in zip((self.pt.table, self.pt.lens, self.pt.refcount, self.cache.pages), self.kept):
            have.copy_(kept)

    def run(self):
        kda = self.kda
        if self.op == "compact":
            kda.kda_pages_compact(self.pt, self.cache, self.pws, self.st)
        elif self.op == "truncate":
            kda.kda_pages_truncate(self.pt, *self.arrays, self.pws, self.st)
        else:
            getattr(kda, "kda_pages_" + self.op)(self.pt, self.cache, *self.arrays, self.pws, self.st)
        for layer in range(2):
            kda.kda_latent_decode(self.cache, layer, self.pt, None, self.cu, 1, self.q, self.out[layer], self.lse[layer],
                                  192 ** -0.5, self.dws, self.st)

    def verify(self):
        """The outputs are those of the table, the lengths and the pages as they are now."""
        from tests.latent_testutil import F64, attend, check
        assert int(self.st.item()) == 0
        for layer in range(2):
            for b in range(ROWS):
                n = int(self.pt.lens[b])
                pos = torch.arange(n, device="cuda")
                kv = self.cache.pages[layer, self.pt.table[b].long()[pos // PAGE], pos % PAGE].to(F64)
                seen = torch.ones(H, n, dtype=torch.bool, device="cuda")
                o, l, to, tl = attend(self.q[b].to(F64), kv, kv[:, :RANK], seen, 192 ** -0.5, torch.bfloat16)
                check(self.out[layer, b], o, to, f"out of row {b}, layer {layer}")
                check(self.lse[layer, b], l, tl, f"lse of row {b}, layer {layer}")


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("op", ["compact", "fork", "truncate", "reserve"])
def test_pool_operation_directly_followed_by_decode(op, captured):
    s = Step(op, seed=len(op))
    s.run()
    torch.cuda.synchronize()
    s.verify()
    moved = not torch.equal(s.pt.table, s.kept[0])
    assert moved
    g = torch.cuda.CUDAGraph()
    if captured:
        s.restore()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            s.run()
    for _ in range(10):
        s.restore()
        s.out.fill_(-7)
        # decode the table as it was first: its lines are on the SMs when the operation changes it
        s.kda.kda_latent_decode(s.cache, 0, s.pt, None, s.cu, 1, s.q, s.out[0], s.lse[0], 192 ** -0.5, s.dws, s.st)
        g.replay() if captured else s.run()
        torch.cuda.synchronize()
        s.verify()
