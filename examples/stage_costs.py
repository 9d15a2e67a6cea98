"""The work of a pipeline's last stage, timed, and what the schedules make of it.

A small stage of residual blocks and a loss head runs its microbatches on one
GPU in the op order of a 1F1B plan, with everything that a microbatch holds
between its F and its W kept in 8 bits:

    F   every block: its product, the join to the residual stream (with
        checkpoints of y and of the block's output), a checkpoint of the next
        input; then the head's loss
    B   the gradients of activations, last block first (join_backward reads the
        checkpoints)
    W   the gradients of the matrices, added to the microbatches' sums, from the
        checkpointed inputs

F, B and W are timed; the times, as ticks, are then the costs of a P-stage
pipeline of such stages that the schedule evaluator compares under GPipe, 1F1B
and the Zero Bubble schedules, next to the bytes that 1F1B's peak of held
microbatches takes in 8 bits and in bf16.

    python examples/stage_costs.py [--tokens 2048 --width 2048 --vocab 32000 --blocks 2 --stages 8 --microbatches 16]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from pipeline_schedule_simulation_gb300 import binding as B  # noqa: E402
from pipeline_schedule_simulation_gb300 import stage as S  # noqa: E402


class Block:
    """y = alpha x + gate * w_post * norm(h W^T), next h = w_pre * norm(y)."""

    def __init__(self, width, gen):
        def normal(*shape, scale=1.0):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)

        self.matrix = normal(width, width, scale=width ** -0.5)
        self.w_post, self.w_pre = 1 + normal(width, scale=0.1), 1 + normal(width, scale=0.1)
        self.gate = normal(1, width, scale=0.5)
        self.sums = {"matrix": torch.zeros(width, width, device="cuda"), "w_post": torch.zeros(width, device="cuda"),
                     "w_pre": torch.zeros(width, device="cuda"), "gate": torch.zeros(1, width, device="cuda")}


class LastStage:
    """Blocks and the loss head of one stage; `held` has what each microbatch keeps."""

    def __init__(self, width, vocab, blocks, alpha=0.9, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.alpha = alpha
        self.blocks = [Block(width, gen) for _ in range(blocks)]
        self.out = (torch.randn(vocab, width, generator=gen, device="cuda") * width ** -0.5).to(torch.bfloat16)
        self.out_sum = torch.zeros(vocab, width, device="cuda")
        self.held = {}

    def forward(self, mb, x, h, target):
        """F: x is the residual stream and h the normed input that the stage before sends.  Returns the tokens' losses."""
        keep = {"target": target, "blocks": []}
        for b in self.blocks:
            kept_h = S.pack(h)
            r = S.join_forward(x, h @ b.matrix.t(), b.w_post, b.w_pre, b.gate, alpha=self.alpha, keep=True)
            x, h = r["y"], r["h"]
            keep["blocks"].append({"h": kept_h, **{k: r[k] for k in ("kept_y", "kept_f", "rstd_post", "rstd_pre")}})
        keep["h"] = S.pack(h)
        # the head's loss is taken on what its gradients will see
        r = S.head_forward(S.unpack(keep["h"]), self.out, target)
        keep["lse"] = r["lse"]
        self.held[mb] = keep
        return r["loss"]

    def backward(self, mb, scale):
        """B: gradients of the stage's two inputs."""
        keep = self.held[mb]
        keep["scale"] = scale
        dh = S.head_backward(S.unpack(keep["h"]), self.out, keep["target"], keep["lse"], scale=scale, outputs=("dx",))["dx"]
        dy = None
        for b, k in zip(reversed(self.blocks), reversed(keep["blocks"])):
            r = S.join_backward(dh, dy, k["kept_y"], k["kept_f"], k["rstd_post"], k["rstd_pre"], b.w_post, b.w_pre, b.gate,
                                alpha=self.alpha)
            for name in ("w_post", "w_pre", "gate"):
                b.sums[name] += r["d" + name]
            k["df"] = r["df"]  # what W needs beside the kept input
            dy, dh = r["dx"], r["df"] @ b.matrix
        return dy, dh

    def weights(self, mb):
        """W: gradients of the matrices, added to the sums; the microbatch is held no longer."""
        keep = self.held.pop(mb)
        for b, k in zip(self.blocks, keep["blocks"]):
            S.weight_grad(k["df"], k["h"], add=b.sums["matrix"], out=b.sums["matrix"])
        S.head_backward(S.unpack(keep["h"]), self.out, keep["target"], keep["lse"], scale=keep["scale"], outputs=("dw",),
                        add=True, out={"dw": self.out_sum})

    def held_bytes(self, mb):
        """Bytes of the activations that a microbatch keeps after its F: in 8 bits, and as they would be in bf16."""
        k = self.held[mb]
        packed = [k["h"]] + [p for b in k["blocks"] for p in (b["h"], b["kept_y"], b["kept_f"])]
        return sum(p.nbytes for p in packed), sum(2 * p.shape[0] * p.shape[1] for p in packed)


def run_1f1b(stage, inputs, targets, stages, device, scale):
    """Runs the microbatches in the op order of one device of a 1F1B plan; returns the losses, the gradients that go
    to the stage before, and the F, B and W times in ms."""
    ops, peak, _ = B.Plan("1f1b", stages, len(inputs)).tables()
    kinds, _, mbs = B.op_fields(ops[device])
    losses, grads, times = [None] * len(inputs), [None] * len(inputs), {"F": [], "B": [], "W": []}

    def timed(kind, f, *a):
        t = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t[0].record()
        r = f(*a)
        t[1].record()
        times[kind].append(t)
        return r

    for kind, mb in zip(kinds.tolist(), mbs.tolist()):
        if kind == 0:
            losses[mb] = timed("F", stage.forward, mb, *inputs[mb], targets[mb])
        else:
            grads[mb] = timed("B", stage.backward, mb, scale)
            timed("W", stage.weights, mb)
        assert len(stage.held) <= int(peak[device])
    failed = S.wait_failure()  # waits for the device
    if failed:
        raise RuntimeError(f"a kernel gave up waiting (record {failed:#x}): the results are wrong")
    return losses, grads, {k: sorted(a.elapsed_time(b) for a, b in v)[len(v) // 2] for k, v in times.items()}


def schedules(f, b, w, stages, microbatches):
    """Makespan in ticks and bubble of the schedules at these costs (ticks of one stage)."""
    def table(v):
        return torch.full((stages * microbatches,), max(1, round(v)), dtype=torch.int32, device="cuda")

    strides = (0, microbatches, 1)
    out = {}
    for name in ("gpipe", "1f1b"):
        out[name] = B.evaluate(name, stages, microbatches, 1, table(f), table(b + w), strides, 1)
    for name in ("zb1p", "zb2p"):
        out[name] = B.evaluate_zb(name, stages, microbatches, table(f), table(b), table(w), strides, 1)
    torch.cuda.synchronize()
    return {k: (int(r["makespan"][0]), int(r["bub_num"][0]) / int(r["bub_den"][0]), r["peak"].flatten().tolist())
            for k, r in out.items()}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--stages", type=int, default=8)
    ap.add_argument("--microbatches", type=int, default=16)
    a = ap.parse_args(argv)
    stage = LastStage(a.width, a.vocab, a.blocks)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    normal = lambda: torch.randn(a.tokens, a.width, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    inputs = [(normal(), normal()) for _ in range(a.microbatches)]
    targets = [torch.randint(0, a.vocab, (a.tokens,), generator=gen, device="cuda") for _ in inputs]
    scale = 1 / (a.tokens * a.microbatches)
    run_1f1b(stage, inputs, targets, a.stages, 0, scale)  # the first run builds plans and loads kernels
    losses, _, ms = run_1f1b(stage, inputs, targets, a.stages, 0, scale)
    print(f"stage of {a.blocks} blocks of width {a.width} and a head of {a.vocab}: {a.tokens} tokens take "
          + ", ".join(f"{k} {v * 1e3:.0f} us" for k, v in ms.items())
          + f"; mean loss {torch.stack(losses).mean().item():.4f}")
    stage.forward(0, *inputs[0], targets[0])
    eight, sixteen = stage.held_bytes(0)
    stage.held.clear()
    for name, (ticks, bubble, peak) in schedules(*(ms[k] * 1e3 for k in "FBW"), a.stages, a.microbatches).items():
        print(f"{name:6s} {a.stages} stages, {a.microbatches} microbatches: makespan {ticks / 1e3:.2f} ms, bubble {bubble:.1%}, "
              f"most held {max(peak)} microbatches = {max(peak) * eight / 1e6:.0f} MB in 8 bits ({max(peak) * sixteen / 1e6:.0f} "
              "MB in bf16)")


if __name__ == "__main__":
    main()
