"""Sizes at which the linear layer's bf16 products take each of their tiles: (product, M, K, N, tile,
reduction ranges).  The products' outputs and reduction: "fwd" M x N over K, "dX" M x K over N, "dW"
N x K over M.  Every tile with an odd and an even number of 64-element stages, more than four, the
last one short; the remainders of M and N leave part of a tile."""

PIPELINED = [
    ("fwd", 2890, 264, 2968, "256x256", 1), ("fwd", 2890, 376, 2965, "256x256", 1),
    ("fwd", 2437, 328, 2488, "256x128", 1), ("fwd", 2437, 264, 2485, "256x128", 1),
    ("fwd", 100, 264, 38392, "ring2", 1), ("fwd", 100, 328, 38389, "ring2", 1),
    ("fwd", 500, 264, 520, "ring4", 1), ("fwd", 500, 328, 517, "ring4", 1),
    ("fwd", 1000, 40000, 1016, "256x256", 16), ("fwd", 1240, 8192, 1656, "256x128", 3),
    ("dX", 2890, 2968, 264, "256x256", 1), ("dX", 2890, 2968, 376, "256x256", 1),
    ("dX", 2437, 2488, 328, "256x128", 1), ("dX", 2437, 2488, 264, "256x128", 1),
    ("dX", 100, 38392, 264, "ring2", 1), ("dX", 100, 38392, 328, "ring2", 1),
    ("dX", 500, 520, 264, "ring4", 1), ("dX", 500, 520, 328, "ring4", 1),
    ("dX", 1000, 1016, 40000, "256x256", 16), ("dX", 1240, 1656, 8192, "256x128", 3),
    ("dW", 261, 2968, 2896, "256x256", 1), ("dW", 383, 2968, 2896, "256x256", 1),
    ("dW", 325, 2488, 2440, "256x128", 1), ("dW", 257, 2488, 2440, "256x128", 1),
    ("dW", 261, 38392, 104, "ring2", 1), ("dW", 325, 38392, 104, "ring2", 1),
    ("dW", 261, 520, 504, "ring4", 1), ("dW", 325, 520, 504, "ring4", 1),
    ("dW", 40001, 1016, 1000, "256x256", 16), ("dW", 8190, 1656, 1240, "256x128", 3),
]

# rows off 16-byte lines (an operand's row length no multiple of 8 elements) in 128 x 128 staged
# tiles: elements loaded one by one, and four by four where every row length is a multiple of 4
STAGED = [
    ("fwd", 2890, 331, 2965, 1), ("fwd", 2890, 332, 2968, 4),
    ("dX", 2890, 2965, 331, 1), ("dX", 2890, 2964, 332, 4),
    ("dW", 331, 2965, 2890, 1), ("dW", 331, 2964, 2892, 4),
]


def outputs_and_reduction(product, M, K, N):
    return {"fwd": (M, N, K), "dX": (M, K, N), "dW": (N, K, M)}[product]
