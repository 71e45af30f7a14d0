"""GB300-native (sm_103a) hot path of a LatentMoE sparse expert layer.

The compute lives in libmoe.so (CUDA, C ABI declared in include/moe.h);
`_lib` binds it with ctypes under the same names, `layer` strings the calls
into a full forward / backward, `route` is its routing with scores and groups, `norm` the
norm before it, `linattn` and `scan` are the sequence mixers beside it, `optim` the optimizer step on their gradients, `inputs` draws the seeded synthetic inputs.
Importing the package does not load the library; the first call does, and it
raises if libmoe.so has not been built.
"""
__all__ = ["_lib", "inputs", "layer", "linattn", "norm", "optim", "route", "scan", "build"]
