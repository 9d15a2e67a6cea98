"""GB300-native batched evaluator of pipeline-parallel training schedules.

GPipe (and its first-in-first-out variant), synchronous 1F1B (PipeDream-Flush),
interleaved 1F1B and the Zero Bubble schedules ZB1P / ZB2P: per-device op
order, every op's start/end tick by max-plus longest path, makespan, per-stage
busy/idle ticks, the exact bubble fraction and the peak count of held
activations, for thousands to millions of instances per call; plus GPU
searches over contiguous layer-to-stage partitions (seeded, exhaustive, and
interleaved layouts).  And the operators of one pipeline stage, whose time and
held bytes are the costs: the last stage's loss over a large vocabulary,
activation checkpoints in 8 bits, the join of a block to the residual stream.

The compute runs in hand-written CUDA kernels behind the C ABI declared in
``include/ppsched.h`` and ``include/ppstage.h`` (``libppsched.so``); ``binding``
and ``stage`` marshal arguments only.  Importing this package does not load the
library: they do, and fail loudly if it has not been built.
"""
__all__ = ["binding", "stage", "workloads", "sharding", "timeline"]
