"""A state-space layer of a hybrid model, served end to end.

The layer's projected rows go through the short convolution, which leaves x, B and C side by
side; the scan takes them where they lie.  Prompts run first, then tokens one at a time,
with both states updated in place; at the end the whole sequences run once more in one
pass, whose last rows the decoded ones have to agree with.

    python examples/state_space_layer.py --tokens 1500 --steps 16
"""
import argparse
import json
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_11_gb300 as kda  # noqa: E402


class Layer:
    """Heads of P channels with S values of state each, B and C shared by the heads of a group."""

    def __init__(self, H, G, P, S, randn):
        self.H, self.G, self.P, self.S = H, G, P, S
        self.channels = H * P + 2 * G * S
        self.weight = (randn(self.channels, 4) / 2).to(torch.bfloat16)
        self.bias = (randn(self.channels) / 10).to(torch.bfloat16)
        self.A = -1.0 - 15.0 * torch.rand(H, device="cuda")
        self.dt_bias = torch.full((H,), -4.0, device="cuda")
        self.skip = torch.ones(H, device="cuda")
        self.conv = self.state = None

    def run(self, scan, rows, dt, cu):
        rows, self.conv = kda.kda_conv_fwd(rows, self.weight, self.bias, initial_state=self.conv, cu_seqlens=cu,
                                           final_state=self.conv)
        T, n, m = rows.shape[0], self.H * self.P, self.G * self.S
        x, B, C = rows[:, :n].view(T, self.H, self.P), rows[:, n:n + m].view(T, self.G, self.S), rows[:, n + m:].view(T, self.G, self.S)
        out, self.state = scan(x, dt, self.A, B, C, self.skip, self.dt_bias, initial_state=self.state, cu_seqlens=cu,
                               final_state=self.state)
        return out

    def prefill(self, rows, dt, cu):
        return self.run(kda.kda_ssm_fwd, rows, dt, cu)

    def decode(self, rows, dt, cu):
        return self.run(kda.kda_ssm_step, rows, dt, cu)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=1500, help="tokens of each prompt")
    p.add_argument("--steps", type=int, default=16, help="tokens decoded for each sequence")
    p.add_argument("--sequences", type=int, default=4)
    p.add_argument("--heads", type=int, default=16)
    p.add_argument("--groups", type=int, default=2)
    a = p.parse_args(argv)
    torch.manual_seed(0)
    randn = lambda *s: torch.randn(s, device="cuda")  # noqa: E731
    N, T, each = a.sequences, a.tokens, a.tokens + a.steps
    layer = Layer(a.heads, a.groups, 64, 128, randn)
    rows = randn(N, each, layer.channels).to(torch.bfloat16)
    dt = randn(N, each, a.heads).to(torch.bfloat16)
    starts = lambda n: torch.arange(N + 1, dtype=torch.int32, device="cuda") * n  # noqa: E731
    flat = lambda t, i, j: t[:, i:j].reshape(N * (j - i), -1)  # noqa: E731

    out = [layer.prefill(flat(rows, 0, T), flat(dt, 0, T), starts(T)).view(N, T, -1)]
    for t in range(T, each):
        out.append(layer.decode(flat(rows, t, t + 1), flat(dt, t, t + 1), starts(1)).view(N, 1, -1))
    out, state = torch.cat(out, 1).float(), layer.state
    layer.conv = layer.state = None
    whole = layer.prefill(flat(rows, 0, each), flat(dt, 0, each), starts(each)).view(N, each, -1).float()
    status = kda.kda_device_status()
    if status:
        raise kda.KdaError(status, "kda_device_status")
    off = lambda x, y: float((x - y).norm() / y.norm())  # noqa: E731
    report = {"sequences": N, "tokens": each, "outputs_differ": off(out, whole), "states_differ": off(state, layer.state)}
    print(json.dumps(report))
    return report


if __name__ == "__main__":
    main()
