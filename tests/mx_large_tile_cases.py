"""Sizes of the GPU tests of tiles of 256 with an epilogue, of experts' products in them and of weight gradients whose groups have many
stages."""

# rows, columns, depth -> whether a workgroup takes several tiles, whether the output (16 bits) is larger than 32 MB
DENSE = {(4090, 4094, 8100): (False, False), (8190, 4094, 6500): (True, True)}
# activation, type of the bias, of the residual, whether the sums are kept, type of y: every activation on each way out
EPILOGUES = [(None, "bf16", None, False, "bf16"), ("relu", "f32", None, False, "f16"), ("silu", None, None, False, "bf16"),
             ("gelu", "bf16", None, False, "bf16"), ("gelu_tanh", "f16", None, False, "f16"),
             (None, None, "bf16", False, "bf16"), ("silu", "bf16", "f32", False, "bf16"), ("relu", "bf16", "f16", False, "f32"),
             (None, "f32", None, True, "bf16"), ("relu", None, None, True, "f32"), ("silu", "bf16", None, True, "bf16"),
             ("gelu", "bf16", None, True, "f16"), ("gelu_tanh", "bf16", None, True, "bf16"),
             ("gelu", "f16", "bf16", True, "bf16"), ("gelu_tanh", None, "f32", True, "bf16"), (None, None, None, False, "f32")]
# rows of each expert, columns, depth; (in front, behind) rows of no expert
GROUPED = [((4000, 0, 1, 255, 2300, 744), 4094, 4352, (0, 0)), ((3333, 257, 3401), 8190, 4352, (5, 304)),
           ((256, 3584, 3460), 4100, 9000, (0, 0))]
GROUPED_EPILOGUES = [(None, "bf16", None, "bf16"), ("relu", "bf16", None, "f16"), ("silu", None, None, "bf16"), ("gelu", "f32", None, "bf16"),
                     ("gelu_tanh", "bf16", None, "bf16"), ("silu", "bf16", "bf16", "bf16"), ("gelu_tanh", "f16", "f32", "f32")]
# rows of each group, with one to five stages of 256 of them in every order; (in front, behind); rows and columns of a gradient
GRADIENTS = [((1100, 0, 513, 1, 257, 700, 255), (0, 0), 4096, 2560), ((255, 700, 257, 1, 1024, 513, 0, 1100), (3, 40), 4098, 2570),
             ((1, 513, 512, 1100, 256, 0, 700), (0, 9), 4095, 2559)]
# rows, columns, depth, groups of a product in tiles of 128; rows, rows and columns of a gradient, groups
MANY_GROUPS = [(40_000, 1024, 1024, 384), (40_000, 1026, 1000, 512), (30_001, 1500, 544, 449)]
MANY_GRADIENTS = [(3000, 130, 136, 384), (2600, 128, 264, 512)]
