"""What the operators of a serving step over a paged cache do at their edges: requests over
their limits, scales far apart, far positions, paths that only some sizes take, faults."""
import ctypes

STRUCTS = ("PlanParams", "RotaryParams", "AppendParams", "GatherParams", "DecodeParams", "PrefillParams")


def test_packed_parameters_fill_the_structs(lib):
    """The bytes that the calls pass are as long as the C struct, which may be copied as a whole."""
    for cls in (getattr(lib, name) for name in STRUCTS):
        args = [i + 0.5 if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(cls._fields_)]
        packed = lib._packer(cls)(*args)
        assert len(packed) == ctypes.sizeof(cls) and packed == bytes(cls(*args)), cls.__name__
