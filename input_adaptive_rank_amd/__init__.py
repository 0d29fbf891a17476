"""DyRA layer forward for AMD MI355X (gfx950).

Submodules:
  synth  -- seeded synthetic inputs (no method arithmetic)
  dyra   -- ctypes binding of the C-ABI library libdyra.so (loaded lazily)
  adapters       -- low-rank adapters of many requests, forward and backward
  block_norm     -- norms around a block with its gate and residual scale
  adapted_block  -- the layer, adapters and norms run together
"""
