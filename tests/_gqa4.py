"""A 4-bit grouped-query cache for tests: pools on the CPU, their values in float64 and the library's handle."""
import numpy as np
import torch

from oracle import gqa_oracle as O

BF, HF, F8 = torch.bfloat16, torch.float16, torch.float8_e4m3fn


def lay(x, token_major):
    return x.transpose(1, 2).contiguous().transpose(1, 2) if token_major else x


def to_device(x):
    """A copy on the GPU with the strides of x ([pages, heads, page, .] pools: either order of heads and slots)."""
    if x is None:
        return None
    if x.dim() == 4 and not x.is_contiguous():
        return x.transpose(1, 2).cuda().transpose(1, 2)
    return x.cuda()


class Cache4:
    """`rows` request rows with room for `slots` slots each in a pool of shuffled pages; pages that nobody owns hold
    NaN blocks.  Block scales of either sign of exponent, down to e4m3's subnormals."""

    def __init__(self, q=BF, hkv=2, dim=64, page=16, rows=3, slots=100, seed=0, token_major=False, scaled=True,
                 wide_scales=False):
        self.qt, self.hkv, self.dim, self.page = q, hkv, dim, page
        self.width = -(-slots // page)
        self.gen = torch.Generator().manual_seed(seed)
        pages = rows * self.width + 3
        order = torch.randperm(pages, generator=self.gen)
        self.table = order[: rows * self.width].view(rows, self.width).to(torch.int32).contiguous()
        for pool in ("k", "v"):
            codes = torch.randint(0, 256, (pages, hkv, page, dim // 2), generator=self.gen, dtype=torch.uint8)
            blocks = 0.2 + 0.3 * torch.rand(pages, hkv, page, dim // 16, generator=self.gen)
            if wide_scales:
                blocks = blocks * torch.exp2(torch.randint(-9, 2, blocks.shape, generator=self.gen).float())
            blocks = blocks.to(F8).view(torch.uint8)
            blocks[order[rows * self.width:]] = 0x7f
            setattr(self, pool, lay(codes, token_major))
            setattr(self, pool + "b", lay(blocks, token_major))
        self.ks = self.vs = None
        if scaled:
            self.ks, self.vs = (0.5 + torch.rand(hkv, generator=self.gen) for _ in range(2))

    def poison(self, lens, rows=None):
        """Blocks without a value behind every request's last row."""
        for b, n in enumerate(lens):
            r = b if rows is None else rows[b]
            for s in range(n, self.width * self.page):
                p, o = int(self.table[r, s // self.page]), s % self.page
                self.kb[p, :, o] = self.vb[p, :, o] = 0xff if s % 2 else 0x7f

    def query(self, batch, heads, spread=1.0):
        return (torch.randn(batch, heads, self.dim, generator=self.gen) * spread).to(self.qt)

    def handle(self, A):
        for name in ("k", "v", "kb", "vb", "table", "ks", "vs"):
            setattr(self, name + "_d", to_device(getattr(self, name)))
        return A.make_gqa_cache(self.k_d, self.v_d, self.table_d, k_scale=self.ks_d, v_scale=self.vs_d,
                                k_blocks=self.kb_d.view(F8), v_blocks=self.vb_d.view(F8))

    def oracle(self):
        return {"k": O.e2m1_values(self.k.numpy(), self.kb.numpy()), "v": O.e2m1_values(self.v.numpy(), self.vb.numpy()),
                "table": self.table.numpy(), "k_scale": None if self.ks is None else self.ks.double().numpy(),
                "v_scale": None if self.vs is None else self.vs.double().numpy()}


def pack(x, scale):
    """The oracle's codes and block scales of rows x [..., KV heads, D] as tensors; scale: [KV heads] or None."""
    s = np.float32(1) if scale is None else scale.numpy()[:, None]
    codes, blocks = O.e2m1_pack(x.float().numpy(), s)
    return torch.from_numpy(codes), torch.from_numpy(blocks)
