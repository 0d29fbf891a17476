"""DyRA layer forward for AMD MI355X (gfx950).

Submodules:
  synth  -- seeded synthetic inputs (no method arithmetic)
  dyra   -- ctypes binding of the C-ABI library libdyra.so (loaded lazily)
  adapters       -- low-rank adapters of many requests, forward and backward
  block_norm     -- norms around a block with its gate and residual scale
  q4             -- projections with 4-bit weights and group scales
  vocab_loss     -- softmax cross entropy over a vocabulary, with its gradients
  adapted_block  -- these run together: a short fine-tuning, then single tokens
"""
