/* What the Python calls ask about a tensor. */
#pragma once

#include <Python.h>
#include <stdint.h>

typedef struct {
    void* ptr;
    const int64_t *shape, *stride;
    int ndim, type;       /* type: index into binding.c's types, -1 none of them */
    int device;           /* of a CUDA tensor, else -1 */
    int contiguous;
} TensorInfo;

#ifdef __cplusplus
extern "C"
#endif
int pa_tensor_info(PyObject* o, TensorInfo* out)
#ifdef __cplusplus
    noexcept
#endif
    ;
