"""MI355X (gfx950) implementation of FlashOptim's fused compressed optimizer
step ("FlashOptim: Optimizers for Memory Efficient Training").

* flashopt.py  -- the thin ctypes binding of the C-ABI HIP library
  (include/flashopt.h; kernels in csrc/, built in-tree by build.py);
* optim.py     -- drop-in FlashAdamW / FlashSGD / FlashLion (torch.optim API,
  compressed checkpoints, gradient release, per-group compression switch,
  HIP-graph capture);
* ablations.py -- the codec studies (weight rebuild error, companding,
  training without companding) and the distillation study (a teacher in 8
  bits) run through the library;
* losses.py    -- losses over rows of logits with their gradients: log
  probabilities of given tokens, entropy, top alternatives, distillation
  (include/flashopt_lm.h);
* int8.py      -- a frozen model's weights in 8 bits and the linear layer over
  them, from a matrix or from the optimizer's state (include/flashopt_lm.h);
* workloads.py -- synthetic parameter-list shapes and seeded input draws for
  the tests and the benchmark.
"""
