"""Sizes of the dense product that between them select every kernel it has
(test_linear_plan.py sees to that)."""

_PLAIN = [(1001, 264, 520), (1001, 264, 1032),    # small tiles; their parts joined
          (5003, 1544, 520), (6001, 2008, 520), (5003, 2824, 520)]  # 192, 224, 256 wide
# (T, N, C, activation)
FORWARD = ([(*s, act) for act in ("none", "silu", "gelu") for s in _PLAIN]
           + [(777, 264, 520, "swiglu"), (777, 264, 1032, "swiglu"), (5003, 776, 520, "swiglu"),
              (777, 7176, 520, "swiglu")]
           # long sums
           + [(2001, 6136, 2056, "none"), (8203, 7176, 2056, "none"), (8203, 1544, 7176, "gelu"),
              (8203, 2056, 7176, "swiglu")])
STREAMED = [(T, N, C, act) for act in ("none", "silu", "gelu", "swiglu")
            for T, N, C in ((13, 72, 1032), (16, 4104, 1032), (100, 264, 520), (61, 2056, 264))]
# (T, N, C): gradients of the rows and of the weights
GRADIENTS = [(777, 264, 520), (1001, 264, 520), (777, 1032, 520),  # small tiles, joined ones
             (777, 7176, 1032), (777, 2824, 4104), (777, 7176, 4104),  # the weights' large tiles
             (1993, 520, 4104), (3001, 520, 4104), (5003, 520, 2824),  # the rows'
             (8203, 4104, 7176)]
