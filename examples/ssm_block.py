"""A state space layer served end to end: packed prompts, then token by token.

The layer is the usual one: an input projection to [z | x | B | C | dt], the short
causal convolution with SiLU over [x | B | C], the selective state space scan with
its gate, and an output projection.  No tensor is copied between them: the
convolution and the scan read column ranges of the projection's output, and the
state pools that the prompts fill are the ones that the single tokens update.

    python examples/ssm_block.py [--steps 8]
"""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_kk_gb300 as gdn  # noqa: E402


class SsmBlock:
    """One layer's weights; its states live in pools that the caller owns."""

    def __init__(self, model=1024, heads=32, head_dim=64, groups=1, state=128, width=4, seed=0,
                 dtype=torch.bfloat16, device="cuda"):
        self.H, self.V, self.G, self.K, self.W = heads, head_dim, groups, state, width
        self.inner, self.channels = heads * head_dim, heads * head_dim + 2 * groups * state
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(shape, generator=gen) * std).to(device)

        self.w_in = normal(self.inner + self.channels + heads, model, std=model ** -0.5).to(dtype)
        self.w_out = normal(model, self.inner, std=self.inner ** -0.5).to(dtype)
        self.conv_w = normal(self.channels, width, std=0.5).to(dtype)
        self.conv_b = normal(self.channels, std=0.1).to(dtype)
        self.A_log = torch.linspace(1, 16, heads, device=device).log()
        self.D = torch.ones(heads, device=device)
        self.dt_bias = normal(heads, std=0.5) - 3

    def pools(self, slots):
        """Zeroed states of ``slots`` requests: the convolution's last rows, the scan's h."""
        dev, dt = self.w_in.device, self.w_in.dtype
        return (torch.zeros((slots, self.W - 1, self.channels), dtype=dt, device=dev),
                torch.zeros((slots, self.H, self.V, self.K), dtype=torch.float32, device=dev))

    def _project(self, u):
        z, xbc, dt = F.linear(u, self.w_in).split([self.inner, self.channels, self.H], -1)
        return z.unflatten(-1, (self.H, self.V)), xbc, dt

    def _split(self, xbc):
        n = self.G * self.K
        x, Bm, Cm = xbc.split([self.inner, n, n], -1)
        return (x.unflatten(-1, (self.H, self.V)), Bm.unflatten(-1, (self.G, self.K)),
                Cm.unflatten(-1, (self.G, self.K)))

    def prompts(self, u, cu_seqlens, pools, slots):
        """u [1,T,model]: packed prompts, prompt n in tokens cu_seqlens[n]..[n+1].
        Leaves their states in the pools' slots and returns [1,T,model]."""
        z, xbc, dt = self._project(u)
        xbc, rows = gdn.short_conv_fwd(xbc, self.conv_w, self.conv_b, cu_seqlens=cu_seqlens)
        x, Bm, Cm = self._split(xbc)
        y, h = gdn.ssm_chunk_fwd(x, dt, self.A_log, Bm, Cm, D=self.D, z=z, dt_bias=self.dt_bias,
                                 cu_seqlens=cu_seqlens)
        pools[0][slots.long()], pools[1][slots.long()] = rows, h
        return F.linear(y.flatten(2), self.w_out)

    def tokens(self, u, pools, slots):
        """u [B,T,model]: the next T = 1..4 tokens of the requests in ``slots``."""
        z, xbc, dt = self._project(u)
        xbc = gdn.short_conv_decode(xbc, self.conv_w, pools[0], self.conv_b, slot_indices=slots)
        x, Bm, Cm = self._split(xbc)
        y = gdn.ssm_decode(x, dt, self.A_log, Bm, Cm, pools[1], D=self.D, z=z,
                           dt_bias=self.dt_bias, slot_indices=slots)
        return F.linear(y.flatten(2), self.w_out)


def main(steps=8, lengths=(300, 1, 77, 640)):
    """Serve ``steps`` tokens of each prompt and compare every output with the one that
    the whole sequence, taken as a prompt, has in its place: returns the largest
    difference over the outputs' root mean square."""
    block = SsmBlock()
    gen = torch.Generator().manual_seed(1)
    u = [torch.randn((n + steps, block.w_in.shape[1]), generator=gen).to(block.w_in) for n in lengths]

    def pack(seqs):
        ends = torch.tensor([0] + [len(s) for s in seqs]).cumsum(0)
        return torch.cat(seqs)[None], ends.to(torch.int32).cuda()

    slots = torch.tensor([5, 0, 3, 6], dtype=torch.int32, device="cuda")
    pools, whole_pools = block.pools(8), block.pools(8)
    packed, cu = pack(u)
    whole = block.prompts(packed, cu, whole_pools, slots)[0].split([len(s) for s in u])

    packed, cu = pack([s[:n] for s, n in zip(u, lengths)])
    got = [list(y.unbind(0)) for y in block.prompts(packed, cu, pools, slots)[0].split(lengths)]
    for t in range(steps):
        step = torch.stack([s[n + t] for s, n in zip(u, lengths)])[:, None]
        for seq, y in zip(got, block.tokens(step, pools, slots)):
            seq.append(y[0])

    torch.cuda.synchronize()
    status = gdn.gdn_check_device_error()
    if status != gdn.Status.OK:
        raise RuntimeError(f"device status {status.name}")
    rms = torch.cat(list(whole)).float().square().mean().sqrt()
    worst = max((torch.stack(g).float() - w.float()).abs().max() for g, w in zip(got, whole))
    return float(worst / rms)


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=8, help="tokens served after each prompt")
    print(f"largest difference / RMS: {main(parser.parse_args().steps):.2e}")
